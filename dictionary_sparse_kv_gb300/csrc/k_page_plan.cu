// Block tables, positions and slots of one step's new tokens.
//
// With n_b = max(add_b, 0), len_b the cached length and P the page size:
//   starts_b = sum_{c<b} n_c                     (rows of the step's tokens)
//   back_b   = ceil(len_b / P) for ended requests (pages returned)
//   need_b   = ceil((len_b + n_b) / P) - ceil(len_b / P)
// and the three prefix sums over the requests decide everything else: page m
// of the step belongs to the request whose prefix of needs holds m, row t to
// the request whose prefix of rows holds t, and both find it by bisection, so
// a prompt of thousands of tokens is spread over the threads like thousands
// of single tokens.  A page taken from the part of the free list that ended
// requests return in this very step is read from its old place in the block
// table, so nothing waits for the list.
//
// A call has to read 8 bytes a request and to write 8 bytes a row: always
// latency.  Few rows: one block does all of it.  Many rows: every block of a
// grid repeats the scan (cheaper than to wait for one that does it) and takes
// an even part of the pages and rows; the lengths and the count, which may be
// updated in place and which every block reads, are written by a last block
// launched behind the grid.  16 single tokens: 3.4 us; 1000 requests with 190000
// rows: 9.5 us.
#include "paged.cuh"

namespace fadkv {
namespace {

// Rows and requests that one block takes: 128 threads where there are few
// (barriers and scans take less than those of 1024), else 1024 threads.
constexpr int kFew = 512;
constexpr int kOneBlock = 4096;
constexpr int kGridThreads = 1024;
constexpr int kGridBlocks = 152;

enum Part { kAll, kGrid, kLast };      // a whole plan; the parts of a plan over a grid

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((long long)tokens + (1 << shift) - 1) >> shift); }

// Largest i in [0, n) with pre[i] <= v, for an ascending pre with pre[0] <= v.
__device__ __forceinline__ int owner(const int* pre, int n, int v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int saturate(long long v) { return v > 0x7fffffffll ? 0x7fffffff : (int)v; }

template <int THREADS, int PART>
__global__ void __launch_bounds__(THREADS)
page_plan_kernel(PlanArgs a)
{
    extern __shared__ int sm[];
    int* st = sm;                      // [B + 1] prefix of rows
    int* nd = st + a.B + 1;            // [B + 1] prefix of needed pages
    int* bk = nd + a.B + 1;            // [B + 1] prefix of returned pages
    int* ln = bk + a.B + 1;            // [B] the served requests' lengths, -1 otherwise
    __shared__ int s_taken, s_refused;
    __shared__ long long s_part[3][THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.B;
    const int first = PART == kGrid ? blockIdx.x * THREADS + tid : tid;       // pages and rows first, first + step, ...
    const int step = PART == kGrid ? gridDim.x * THREADS : THREADS;
    const int most = a.max_pages << a.shift;
    const int each = (B + THREADS - 1) / THREADS, b0 = min(B, tid * each), b1 = min(B, b0 + each);
    // the last block starts behind every grid block's wait: what the plan reads is complete for it too
    if (PART != kLast) pdl_begin();
    if (tid == 0) s_taken = s_refused = 0;

    auto length = [&](int b) { return min(max(a.lengths[b], 0), most); };
    // rows, needed and returned pages of a request
    auto item = [&](int b, long long (&v)[3]) {
        const int len = length(b), add = a.add[b];
        v[0] = max(add, 0);
        v[1] = add > 0 && (long long)len + add <= most ? pages_of(len + add, a.shift) - pages_of(len, a.shift) : 0;
        v[2] = add < 0 ? pages_of(len, a.shift) : 0;
    };
    const int count = min(max(*a.free_count, 0), a.num_pages);
    long long v[3], mine[3] = {0, 0, 0}, at[3], total[3];
    for (int b = b0; b < b1; ++b) {
        item(b, v);
#pragma unroll
        for (int k = 0; k < 3; ++k) mine[k] += v[k];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        at[k] = mine[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, at[k], o);
            if (lane >= o) at[k] += y;
        }
        if (lane == 31) s_part[k][warp] = at[k];
    }
    __syncthreads();
    constexpr int W = THREADS / 32;
    if (warp == 0) {                                   // the warps' sums: their prefix sums, the whole one last
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            long long x = lane < W ? s_part[k][lane] : 0;
#pragma unroll
            for (int o = 1; o < W; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane < W) s_part[k][lane] = x;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        at[k] -= mine[k];
        if (warp > 0) at[k] += s_part[k][warp - 1];
        total[k] = s_part[k][W - 1];
    }
    const int returned = (int)min(total[2], (long long)(a.num_pages - count)), F = count + returned;
    int taken = 0, refused = 0;
    for (int b = b0; b < b1; ++b) {
        const int len = length(b), add = a.add[b];
        item(b, v);
        const bool fits = (long long)len + max(add, 0) <= most && at[0] + v[0] <= a.max_tokens;
        const bool served = add > 0 && fits && (v[1] == 0 || at[1] + v[1] <= F);
        st[b] = saturate(at[0]);
        nd[b] = saturate(at[1]);
        bk[b] = saturate(at[2]);
        ln[b] = served ? len : -1;
        if (served && v[1] > 0) taken = (int)(at[1] + v[1]);
        refused += add > 0 && !served;
        if (PART == kAll || (PART == kGrid && blockIdx.x == 0)) a.starts[b] = st[b];
#pragma unroll
        for (int k = 0; k < 3; ++k) at[k] += v[k];
    }
    if (taken) atomicMax(&s_taken, taken);
    if (refused) atomicAdd(&s_refused, refused);
    if (tid == 0) {
        st[B] = saturate(total[0]);
        nd[B] = saturate(total[1]);
        bk[B] = saturate(total[2]);
        if (PART == kAll || (PART == kGrid && blockIdx.x == 0)) a.starts[B] = st[B];
    }
    __syncthreads();
    taken = s_taken;

    if (PART != kLast) {
        // entry i of the free list after the returns
        auto entry = [&](int i) {
            if (i < count) return a.free_pages[i];
            const int b = owner(bk, B, i - count);
            return a.table[(size_t)b * a.max_pages + i - count - bk[b]];
        };
        for (int i = first; i < returned; i += step) a.free_pages[count + i] = entry(count + i);
        for (int m = first; m < taken; m += step) {
            const int b = owner(nd, B, m);
            a.table[(size_t)b * a.max_pages + pages_of(ln[b], a.shift) + m - nd[b]] = entry(F - 1 - m);
        }
        const int T = st[B];
        for (int t = first; t < a.max_tokens; t += step) {
            int pos = -1, slot = -1;
            if (t < T) {
                const int b = owner(st, B, t);
                if (ln[b] >= 0) {
                    pos = ln[b] + t - st[b];
                    // a page that the request had, or one taken in this step
                    const int fresh = (pos >> a.shift) - pages_of(ln[b], a.shift);
                    const int page = fresh >= 0 ? entry(F - 1 - nd[b] - fresh) : a.table[(size_t)b * a.max_pages + (pos >> a.shift)];
                    if (page >= 0 && page < a.num_pages) slot = (page << a.shift) + (pos & ((1 << a.shift) - 1));
                }
            }
            a.positions[t] = pos;
            a.slots[t] = slot;
        }
    }
    if (PART == kGrid) return;
    // nothing of the grid reads the lengths and the count any more
    if (PART == kLast) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int b = b0; b < b1; ++b) {
        const int len = length(b), add = a.add[b];
        a.lengths_out[b] = add < 0 ? 0 : (ln[b] >= 0 ? len + add : len);
    }
    if (tid == 0) {
        *a.free_count_out = F - taken;
        *a.refused = s_refused;
    }
}

template <int THREADS, int PART>
cudaError_t allow_smem(size_t smem)
{
    if (smem <= 48 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(page_plan_kernel<THREADS, PART>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t st)
{
    const size_t smem = (size_t)(4 * a.B + 3) * sizeof(int);
    if (a.B <= kFew && a.max_tokens <= kFew) {
        return launch_pdl(page_plan_kernel<128, kAll>, dim3(1), dim3(128), smem, st, a);
    }
    if (a.max_tokens <= kOneBlock) {
        const cudaError_t e = allow_smem<1024, kAll>(smem);
        if (e != cudaSuccess) return e;
        return launch_pdl(page_plan_kernel<1024, kAll>, dim3(1), dim3(1024), smem, st, a);
    }
    cudaError_t e = allow_smem<kGridThreads, kGrid>(smem);
    if (e == cudaSuccess) e = allow_smem<1024, kLast>(smem);
    if (e != cudaSuccess) return e;
    const int blocks = (a.max_tokens + kGridThreads - 1) / kGridThreads;
    e = launch_pdl(page_plan_kernel<kGridThreads, kGrid>, dim3(blocks < kGridBlocks ? blocks : kGridBlocks),
                   dim3(kGridThreads), smem, st, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_plan_kernel<1024, kLast>, dim3(1), dim3(1024), smem, st, a);
}

}  // namespace fadkv
