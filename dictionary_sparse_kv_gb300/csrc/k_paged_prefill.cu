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
// it.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since
// the last time (p then stays below 2^8, far inside both 16-bit types, and
// o / l is the same), which after the first tiles is rare; the rescale goes
// through registers in the softmax warps.
//
// K and V pages come by TMA, one box a page and 64-element half, through one
// ring of stages; pages outside the pool and pages that no row sees are asked
// for outside the map and arrive as zeros.  Keys that a row does not see are
// masked in registers, in the key tiles where that can happen.  What a seen
// page holds past the tokens that the tile sees may be anything, so its value
// rows are zeroed in shared memory before the product (0 x NaN would be NaN).
//
// Warps: 0 TMA, 1 MMA, 2 TMEM and the zeroing, 4..7 and 8..11 softmax of the
// two tiles.  Every wait is bounded; one that runs out sets
// FADKV_DEV_TIMEOUT in the workspace's first word, and the CTA drains and
// returns.
#include "paged.cuh"
#include "tc_common.cuh"

namespace fadkv {
namespace {

using namespace paged;
using namespace tc;

constexpr int kPreThreads = 384;
constexpr int kRows = 128;                         // (token, head) rows per tile, two tiles per CTA
constexpr int kKeys = 128;                         // keys per tile
constexpr int kFix = 4;                            // barriers of the zeroing, in turn: as many as value stages at least
constexpr int kOkRing = 16;                        // key tiles whose page masks are kept
constexpr float kGrow = 8.f;                       // growth of the maximum (log2) that rescales

template <int D> struct PreCfg {
    static constexpr int NST = D == 128 ? 5 : 8;   // stages of the K / V ring
    static constexpr int TILE = kRows * D * 2;     // bytes of a Q, K or V tile
    static constexpr int bar_off = (2 + NST) * TILE;
    static constexpr int n_bars = 2 * NST + 10 + kFix;
    static constexpr int ok_off = bar_off + n_bars * 8;
    static constexpr int alloc = ok_off + kOkRing * 20 + 16 + 1024;
    static_assert(alloc <= 227 * 1024, "shared memory");
    // TMEM columns.  d = 128: P over the first half of its S (the products of
    // one thread with one shape run in order); d = 64: room for its own.
    static constexpr int S(int q) { return q * 128; }
    static constexpr int O(int q) { return 256 + q * D; }
    static constexpr int P(int q) { return D == 128 ? q * 128 : 384 + q * 64; }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
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

// Two 32-bit values in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Bits 0 .. n-1 set (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

template <typename T, int D>
__global__ void __launch_bounds__(kPreThreads, 1)
paged_prefill_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ PagedArgs a)
{
    using C = PreCfg<D>;
    constexpr int NST = C::NST, HALVES = D / 64, TILE = C::TILE;
    extern __shared__ unsigned char smem_raw[];
    __shared__ int s_b, s_tile;
    __shared__ uint32_t s_taddr;
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sQ = smem_u32(smem), sR = sQ + 2 * TILE, bar0 = sQ + C::bar_off;
    uint32_t* ok_ring = reinterpret_cast<uint32_t*>(smem + C::ok_off);   // [kOkRing][5]: all ok, four words of key bits
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (NST + s); };
    auto sfull = [&](int q) { return bar0 + 8u * (2 * NST + q); };
    auto pvdone = [&](int q) { return bar0 + 8u * (2 * NST + 2 + q); };
    auto qfull = [&](int q) { return bar0 + 8u * (2 * NST + 4 + q); };
    auto pfull = [&](int q, int half) { return bar0 + 8u * (2 * NST + 6 + 2 * q + half); };
    auto fixed = [&](int j) { return bar0 + 8u * (2 * NST + 10 + (j & (kFix - 1))); };
    unsigned long long* status = reinterpret_cast<unsigned long long*>(a.ws);

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int grp = a.grp, B = a.p.B;
    const int gch = min(grp, kRows), chunks = (grp + gch - 1) / gch, tq = kRows / gch;   // tokens per tile
    const int heads = a.p.Hkv * chunks, per_cta = 2 * tq;
    const int hk = (int)(blockIdx.x % heads) / chunks, h0 = (int)(blockIdx.x % chunks) * gch, hn = min(gch, grp - h0);

    auto rows_of = [&](int b) {
        const int s = a.starts[b];
        return s < 0 ? 0 : max(0, min(a.starts[b + 1], a.p.T) - s);
    };
    {
        const int each = (B + kPreThreads - 1) / kPreThreads, b0 = min(B, tid * each), b1 = min(B, b0 + each);
        long long mine = 0, all;
        for (int b = b0; b < b1; ++b) mine += (rows_of(b) + per_cta - 1) / per_cta;
        long long at = block_scan<kPreThreads>(mine, &all);
        const long long u = all - 1 - blockIdx.x / heads;   // a request's last tiles see the most keys: first
        if (u < 0) return;
        if (u >= at && u < at + mine) {
            int b = b0;
            for (long long n; u >= at + (n = (rows_of(b) + per_cta - 1) / per_cta); ++b) at += n;
            s_b = b;
            s_tile = (int)(u - at);
        }
    }
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int q = 0; q < 2; ++q) {
            mbar_init(sfull(q), 1);
            mbar_init(pfull(q, 0), 4);
            mbar_init(pfull(q, 1), 4);
            mbar_init(pvdone(q), 1);
            mbar_init(qfull(q), 128);
        }
        for (int j = 0; j < kFix; ++j) mbar_init(fixed(j), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_taddr)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, s_taddr, 0);

    const int b = __shfl_sync(0xffffffffu, s_b, 0), t0 = __shfl_sync(0xffffffffu, s_tile, 0) * per_cta, start = a.starts[b];
    const int nt = min(per_cta, rows_of(b) - t0);      // tokens of this CTA
    const int nq = nt > tq ? 2 : 1;                    // tiles that hold any
    const int len = clamp_len(a.lengths[b], a);
    // positions by the rows that the request has, those cut off at T included
    const int first = len - (a.starts[b + 1] - start) + t0, last = first + nt - 1;
    const int W = min(a.p.window, 1 << 30), S = min(a.p.sinks, len);

    // key tiles: those of the first tokens, then those of the window (or all)
    const int tiles_to = last >= 0 ? last / kKeys + 1 : 0;
    const int from = W > 0 ? max(0, first - W + 1) / kKeys : 0;
    const int sink_tiles = W > 0 ? min(from, (S + kKeys - 1) / kKeys) : 0;
    const int tiles = __shfl_sync(0xffffffffu, tiles_to > from ? sink_tiles + tiles_to - from : 0, 0);
    auto key0 = [&](int i) { return (i < sink_tiles ? i : i - sink_tiles + from) * kKeys; };
    // whether some row of the CTA sees a key; whether a tile holds keys that none sees
    auto seen = [&](int key) { return key <= last && (W == 0 || key > first - W || key < S); };
    auto ragged = [&](int k0) { return !(k0 + kKeys - 1 <= last && (W == 0 || k0 > first - W || k0 + kKeys <= S)); };

    // Registers: 168 a thread at launch (384 threads, 64512 in all); the four
    // service warps keep 104, the eight softmax warps take 200.
    if (warp == 0) {
        regs_dec();
        // ---------------- K and V pages ----------------
        const int rows = min(1 << a.shift, kKeys), boxes = kKeys / rows * HALVES;   // at most 32
        const int row = lane / HALVES * rows, half = lane % HALVES;
        int issued = 0;
        bool ok = true;
        auto page_of = [&](int i) {
            int page = -1;
            if (i < tiles && lane < boxes) {
                const int key = key0(i) + row;
                // the box is asked for if any of its keys is seen: the first, the last up to `last`, or one of the first tokens
                if (key <= last && (seen(key) || seen(min(key + rows - 1, last))))
                    page = __ldg(a.table + (size_t)b * a.p.max_pages + (key >> a.shift));
                if (page >= a.p.num_pages) page = -1;
            }
            return page;
        };
        int page = page_of(0);
        for (int i = 0; i < tiles && ok; ++i) {
            const int k0 = key0(i), next = page_of(i + 1);
            const uint32_t good = __ballot_sync(0xffffffffu, page >= 0 || lane >= boxes);
            for (int kv = 0; kv < 2 && ok; ++kv) {
                const int s = issued % NST;
                ok = mbar_wait(empty(s), ((uint32_t)(issued / NST) & 1u) ^ 1u, status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    if (kv == 0) {
                        uint32_t* o = ok_ring + (i & (kOkRing - 1)) * 5;
                        o[0] = good == 0xffffffffu;
                        if (good != 0xffffffffu) {
                            for (int w = 0; w < 4; ++w) {
                                uint32_t bits = 0;
                                for (int r = 0; r < 32; r += 8)
                                    if ((good >> ((w * 32 + r) / rows * HALVES)) & 1u) bits |= 0xffu << r;
                                o[1 + w] = bits;
                            }
                        }
                    }
                    mbar_expect_tx(full(s), TILE);
                }
                __syncwarp();
                if (lane < boxes)
                    tma_load_4d(sR + s * TILE + half * (kKeys * 128) + row * 128, kv ? &map_v : &map_k, half * 64,
                                k0 & ((1 << a.shift) - 1) & ~(rows - 1), hk, page >= 0 ? page : a.p.num_pages, full(s));
                ++issued;
            }
            page = next;
        }
        // drain: every issued load lands before the CTA exits
        for (int i = max(0, issued - NST); i < issued; ++i) mbar_wait(full(i % NST), (uint32_t)(i / NST) & 1u, status);
    } else if (warp == 1) {
        regs_dec();
        // ---------------- products ----------------
        // The whole warp walks the tiles, so that descriptors and addresses stay in
        // uniform registers; one thread issues.  (With the walk in one thread alone
        // each product costs about 90 cycles to issue, against 64 to run.)
        if (tiles > 0) {
            constexpr uint32_t kQK = idesc_of<T>(kRows, kKeys, false), kPV = idesc_of<T>(kRows, D, true);
            const bool leader = elect_one();
            bool ok = true;
            int pvs[2] = {0, 0}, qks[2] = {0, 0};
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
            };
            // stage and parity of the next ring entry: K and V in turn
            int st = 0;
            uint32_t ph = 0;
            auto next_entry = [&] {
                if (++st == NST) {
                    st = 0;
                    ph ^= 1u;
                }
            };
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
            // one half of the keys
            auto pv = [&](int q, int stage, int half, bool add) {
                const uint64_t dv = dn0 + (uint64_t)(stage * (TILE >> 4) + half * (kKeys / 2 * 128 >> 4));
                if (leader)
#pragma unroll
                    for (int j = 0; j < kKeys / 32; ++j)
                        mma_ts(tbase + C::O(q), tbase + C::P(q) + (half * (kKeys / 32) + j) * 8, dv + (uint64_t)(j * 2048 >> 4),
                               kPV, add || j > 0 ? 1u : 0u);
            };
            for (int q = 0; q < nq; ++q) wait(qfull(q), 0u);
            wait(full(0), 0u);
            if (ok) {
                fence_after();
                for (int q = 0; q < nq; ++q) qk(q, 0);
                if (leader) mma_commit(empty(0));
                next_entry();
            }
            for (int i = 0; i < tiles && ok; ++i) {
                const int sv = st;
                const uint32_t pv_ph = ph;
                next_entry();                              // now the next tile's K
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (q >= nq || !ok) continue;
                    if (q == 0) {
                        wait(full(sv), pv_ph);
                        wait(fixed(i), (uint32_t)(i / kFix) & 1u);
                    }
                    wait(pfull(q, 0), (uint32_t)i & 1u);
                    if (!ok) break;
                    fence_after();
                    pv(q, sv, 0, i > 0);
                    wait(pfull(q, 1), (uint32_t)i & 1u);
                    if (q == 0 && i + 1 < tiles) wait(full(st), ph);
                    if (!ok) break;
                    fence_after();
                    pv(q, sv, 1, true);
                    if (leader) mma_commit(pvdone(q));
                    ++pvs[q];
                    if (q == nq - 1 && leader) mma_commit(empty(sv));
                    if (i + 1 < tiles) {
                        qk(q, st);
                        if (q == nq - 1 && leader) mma_commit(empty(st));
                    }
                }
                next_entry();
            }
            // drain: the last products of each tile are complete before TMEM is freed
            for (int q = 0; q < 2; ++q) {
                if (qks[q] > 0) mbar_wait(sfull(q), (uint32_t)(qks[q] - 1) & 1u, status);
                if (pvs[q] > 0) mbar_wait(pvdone(q), (uint32_t)(pvs[q] - 1) & 1u, status);
            }
            __syncwarp();
        }
    } else if (warp == 2) {
        regs_dec();
        // ---------------- value rows that no row sees: zeros ----------------
        // Every value tile passes here on its way to the product, so that this
        // warp stays within one round of the ring.
        bool ok = true;
        for (int i = 0; i < tiles && ok; ++i) {
            const int k0 = key0(i), r = 2 * i + 1, s = r % NST;
            ok = mbar_wait(full(s), (uint32_t)(r / NST) & 1u, status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (ragged(k0)) {
                for (int row = 0; row < kKeys; ++row) {
                    if (seen(k0 + row)) continue;
                    // the whole row, so wherever the swizzle puts its 16-byte pieces
                    if (lane < D / 8)
                        *reinterpret_cast<uint4*>(smem + (2 + s) * TILE + (lane / 8) * (kKeys * 128) + row * 128 +
                                                  (lane % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(fixed(i));
        }
    } else if (warp == 3) {
        regs_dec();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---------------- softmax ----------------
        const int q = (warp - 4) >> 2, r = tid & 127;
        if (q < nq) {
            // queries into shared memory (swizzled 128-byte rows), a negative scale's sign and a zero scale with them
            {
                const uint32_t flip = a.p.scale < 0.f ? 0x80008000u : 0u;
                const bool zero = a.p.scale == 0.f;
                const T* qp = (const T*)a.q + (size_t)(hk * grp + h0) * D;
#pragma unroll 8
                for (int j = r; j < kRows * (D / 8); j += 128) {
                    const int row = j / (D / 8), c = j % (D / 8), t = q * tq + row / gch, h = row % gch;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (row / gch < tq && t < nt && h < hn && !zero) {
                        v = __ldg(reinterpret_cast<const uint4*>(qp + (size_t)(start + t0 + t) * a.p.q_stride + h * D) + c);
                        v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
                    }
                    *reinterpret_cast<uint4*>(smem + q * TILE + (c / 8) * (kRows * 128) + swz<128>(row, c & 7)) = v;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(qfull(q));
            }
            const int t = q * tq + r / gch, h = r % gch;
            const bool live = r / gch < tq && t < nt && h < hn;
            const int pos = live ? first + t : -1;
            const int pmin = first + q * tq, pmax = min(last, pmin + tq - 1);
            const float scale = a.p.scale == 0.f ? 1.f : fabsf(a.scale_log2);
            const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int i = 0; i < tiles && ok; ++i) {
                ok = mbar_wait(sfull(q), (uint32_t)i & 1u, status);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_async(lanes + C::S(q) + c * 32, s[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait32(s[c]);
                const int k0 = key0(i);
                const uint32_t* okr = ok_ring + (i & (kOkRing - 1)) * 5;
                // masks only where the tile has keys that some row of the 128 does not see
                if (!(k0 + kKeys - 1 <= pmin && (W == 0 || k0 > pmax - W || k0 + kKeys <= S) && okr[0])) {
                    const bool all_ok = okr[0] != 0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int k = k0 + c * 32;
                        uint32_t bits = low_bits(pos - k + 1);
                        if (W > 0) bits &= ~low_bits(pos - W - k + 1) | low_bits(S - k);
                        if (!all_ok) bits &= okr[1 + c];
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!((bits >> j) & 1u)) s[c][j] = 0xff800000u;
                    }
                }
                float mx = -INFINITY;
                {
                    float x[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        x[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
                        for (int j = 2; j < 32; j += 2)
                            x[c] = max3(x[c], __uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]));
                    }
                    mx = fmaxf(max3(x[0], x[1], x[2]), x[3]) * scale;
                }
                const bool grow = mx > m + kGrow;
                if (__any_sync(0xffffffffu, grow)) {
                    float f = 1.f;
                    if (grow) {
                        f = exp2_fast(m - mx);
                        m = mx;
                        l *= f;
                    }
                    if (i > 0) {
                        ok = mbar_wait(pvdone(q), (uint32_t)(i - 1) & 1u, status);
                        if (!__all_sync(0xffffffffu, ok)) {
                            ok = false;
                            break;
                        }
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
                    tmem_st16(lanes + C::P(q) + c * 16, p);
                    if (c & 1) {                               // half of the keys: the product may begin
                        tmem_st_wait();
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(pfull(q, c >> 1));
                    }
                }
                float x0, x1;
                unpair(add2(sum[0], sum[1]), x0, x1);
                l += x0 + x1;
            }
            if (tiles > 0 && ok) {
                ok = mbar_wait(pvdone(q), (uint32_t)(tiles - 1) & 1u, status);
                ok = __all_sync(0xffffffffu, ok);
                fence_after();
            }
            if (ok) {
                const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
                const size_t row = (size_t)start + t0 + t, head = (size_t)hk * grp + h0 + h;
                uint4* out = reinterpret_cast<uint4*>((T*)a.out + row * a.p.out_stride + head * D);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (tiles > 0) {
                        tmem_ld32(lanes + C::O(q) + c * 32, o);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0u;
                    }
                    if (live)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            auto two = [&](int k) {
                                return Num<T>::pack(__uint_as_float(o[8 * j + 2 * k]) * inv,
                                                    __uint_as_float(o[8 * j + 2 * k + 1]) * inv);
                            };
                            out[c * 4 + j] = make_uint4(two(0), two(1), two(2), two(3));
                        }
                }
                if (live && a.lse) a.lse[row * a.p.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            }
        }
    }

    fence_before();
    __syncthreads();
    if (warp == 2) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512));
    }
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

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t st)
{
    auto k = paged_prefill_kernel<T, D>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, PreCfg<D>::alloc);
    if (e != cudaSuccess) return e;
    CUtensorMap mk, mv;
    if (!pool_map(&mk, a.k, a) || !pool_map(&mv, a.v, a)) return cudaErrorInvalidValue;
    const int gch = a.grp < kRows ? a.grp : kRows, chunks = (a.grp + gch - 1) / gch, tq = kRows / gch;
    const long long tiles = a.p.T / (2 * tq) + a.p.B;
    k<<<(unsigned)(tiles * a.p.Hkv * chunks), kPreThreads, PreCfg<D>::alloc, st>>>(mk, mv, a);
    return cudaGetLastError();
}

}  // namespace

size_t paged_prefill_workspace(const fadkv_paged_params&) { return 256; }

cudaError_t launch_paged_prefill(const PagedArgs& a, cudaStream_t st)
{
    if (a.p.B <= 0 || a.p.T <= 0) return cudaSuccess;
    if (a.p.dtype == FADKV_F16) return a.p.d == 128 ? launch_t<__half, 128>(a, st) : launch_t<__half, 64>(a, st);
    return a.p.d == 128 ? launch_t<__nv_bfloat16, 128>(a, st) : launch_t<__nv_bfloat16, 64>(a, st);
}

}  // namespace fadkv
