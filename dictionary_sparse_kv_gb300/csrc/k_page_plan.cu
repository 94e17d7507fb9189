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
// of single tokens.  One block scans the requests; it has to read 8 bytes a
// request and to write 8 bytes a row, so the small calls are latency (one
// block, one launch) and for many rows a second kernel over the whole grid
// writes positions and slots.
#include "paged.cuh"

namespace fadkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;
// Rows that the scanning block writes itself, in place of a second launch.
constexpr int kRowsInPlan = 4096;

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

__device__ __forceinline__ void write_row(const PlanArgs& a, int t, int b, int pos)
{
    int slot = -1;
    if (pos >= 0) {
        const int page = a.table[(size_t)b * a.max_pages + (pos >> a.shift)];
        if (page >= 0 && page < a.num_pages) slot = (page << a.shift) + (pos & ((1 << a.shift) - 1));
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
}

__global__ void __launch_bounds__(kPlanThreads)
page_plan_kernel(PlanArgs a, int rows_here)
{
    extern __shared__ int sm[];
    int* st = sm;                      // [B + 1] prefix of rows
    int* nd = st + a.B + 1;            // [B + 1] prefix of needed pages
    int* bk = nd + a.B + 1;            // [B + 1] prefix of returned pages; then the served requests' lengths, -1 otherwise
    __shared__ int s_taken, s_refused;
    const int tid = threadIdx.x, B = a.B;
    const int most = a.max_pages << a.shift;
    const int each = (B + kPlanThreads - 1) / kPlanThreads, b0 = min(B, tid * each), b1 = min(B, b0 + each);
    if (tid == 0) s_taken = s_refused = 0;

    auto length = [&](int b) { return min(max(a.lengths[b], 0), most); };
    auto item = [&](int b, long long& n, long long& need, long long& back) {
        const int len = length(b), add = a.add[b];
        n = max(add, 0);
        need = (n > 0 && len + n <= most) ? pages_of((int)(len + n), a.shift) - pages_of(len, a.shift) : 0;
        back = add < 0 ? pages_of(len, a.shift) : 0;
    };
    long long n, need, back, sn = 0, sneed = 0, sback = 0, tn, tneed, tback;
    for (int b = b0; b < b1; ++b) {
        item(b, n, need, back);
        sn += n;
        sneed += need;
        sback += back;
    }
    sn = paged::block_scan<kPlanThreads>(sn, &tn);
    sneed = paged::block_scan<kPlanThreads>(sneed, &tneed);
    sback = paged::block_scan<kPlanThreads>(sback, &tback);
    for (int b = b0; b < b1; ++b) {
        item(b, n, need, back);
        st[b] = saturate(sn);
        nd[b] = saturate(sneed);
        bk[b] = saturate(sback);
        a.starts[b] = st[b];
        sn += n;
        sneed += need;
        sback += back;
    }
    if (tid == 0) {
        st[B] = saturate(tn);
        nd[B] = saturate(tneed);
        bk[B] = saturate(tback);
        a.starts[B] = st[B];
    }
    const int count = min(max(*a.free_count, 0), a.num_pages);
    __syncthreads();
    const int returned = min(bk[B], a.num_pages - count), F = count + returned;
    for (int i = tid; i < returned; i += kPlanThreads) {
        const int b = owner(bk, B, i);
        a.free_pages[count + i] = a.table[(size_t)b * a.max_pages + i - bk[b]];
    }
    __syncthreads();
    for (int b = b0; b < b1; ++b) {
        const int len = length(b), add = a.add[b];
        const bool served = add > 0 && (long long)len + add <= most && st[b + 1] <= a.max_tokens &&
                            (nd[b + 1] == nd[b] || nd[b + 1] <= F);
        bk[b] = served ? len : -1;
        a.lengths_out[b] = add < 0 ? 0 : (served ? len + add : len);
        if (served && nd[b + 1] > nd[b]) atomicMax(&s_taken, nd[b + 1]);
        if (add > 0 && !served) atomicAdd(&s_refused, 1);
        if (!rows_here && add > 0 && st[b] < a.max_tokens) a.positions[st[b]] = served ? len : -1;
    }
    __syncthreads();
    const int taken = s_taken;
    for (int m = tid; m < taken; m += kPlanThreads) {
        const int b = owner(nd, B, m);
        a.table[(size_t)b * a.max_pages + pages_of(bk[b], a.shift) + m - nd[b]] = a.free_pages[F - 1 - m];
    }
    if (tid == 0) {
        *a.free_count_out = F - taken;
        *a.refused = s_refused;
    }
    if (!rows_here) return;
    __syncthreads();
    const int T = st[B];
    for (int t = tid; t < a.max_tokens; t += kPlanThreads) {
        int b = 0, pos = -1;
        if (t < T) {
            b = owner(st, B, t);
            if (bk[b] >= 0) pos = bk[b] + t - st[b];
        }
        write_row(a, t, b, pos);
    }
}

// Rows over the whole grid.  The first row of each request holds its first
// position already (-1 if refused); the thread of that row writes the same
// value again.
__global__ void __launch_bounds__(kRowThreads)
page_rows_kernel(PlanArgs a)
{
    pdl_begin();
    const int t = blockIdx.x * kRowThreads + threadIdx.x;
    if (t >= a.max_tokens) return;
    int b = 0, pos = -1;
    if (t < a.starts[a.B]) {
        b = owner(a.starts, a.B, t);
        const int s = a.starts[b], first = a.positions[s];
        if (first >= 0) pos = first + t - s;
    }
    write_row(a, t, b, pos);
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t st)
{
    const size_t smem = (size_t)3 * (a.B + 1) * sizeof(int);
    const int rows_here = a.max_tokens <= kRowsInPlan;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024)
        e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    page_plan_kernel<<<1, kPlanThreads, smem, st>>>(a, rows_here);
    e = cudaGetLastError();
    if (e != cudaSuccess || rows_here) return e;
    return launch_pdl(page_rows_kernel, dim3((unsigned)((a.max_tokens + kRowThreads - 1) / kRowThreads)),
                      dim3(kRowThreads), 0, st, a);
}

}  // namespace fadkv
