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

constexpr int kRowThreads = 256;
// Rows that the scanning block writes itself, in place of a second launch.
constexpr int kRowsInPlan = 4096;
// A block of 128 threads where requests and rows are few: its barriers and
// scans take less than those of 1024.
constexpr int kFew = 512;

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

__device__ __forceinline__ void write_row(const PlanArgs& a, int t, int pos, int page)
{
    a.positions[t] = pos;
    a.slots[t] = pos >= 0 && page >= 0 && page < a.num_pages ? (page << a.shift) + (pos & ((1 << a.shift) - 1)) : -1;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS)
page_plan_kernel(PlanArgs a, int rows_here)
{
    extern __shared__ int sm[];
    int* st = sm;                      // [B + 1] prefix of rows
    int* nd = st + a.B + 1;            // [B + 1] prefix of needed pages
    int* bk = nd + a.B + 1;            // [B + 1] prefix of returned pages; then the served requests' lengths, -1 otherwise
    __shared__ int s_taken, s_refused;
    __shared__ long long s_part[3][THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.B;
    const int most = a.max_pages << a.shift;
    const int each = (B + THREADS - 1) / THREADS, b0 = min(B, tid * each), b1 = min(B, b0 + each);
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
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        at[k] -= mine[k];
        total[k] = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) at[k] += s_part[k][w];
            total[k] += s_part[k][w];
        }
    }
    for (int b = b0; b < b1; ++b) {
        st[b] = saturate(at[0]);
        nd[b] = saturate(at[1]);
        bk[b] = saturate(at[2]);
        a.starts[b] = st[b];
        if (each > 1) item(b, v);
#pragma unroll
        for (int k = 0; k < 3; ++k) at[k] += each > 1 ? v[k] : mine[k];
    }
    if (tid == 0) {
        st[B] = saturate(total[0]);
        nd[B] = saturate(total[1]);
        bk[B] = saturate(total[2]);
        a.starts[B] = st[B];
    }
    __syncthreads();
    const int returned = min(bk[B], a.num_pages - count), F = count + returned;
    if (returned > 0) {
        for (int i = tid; i < returned; i += THREADS) {
            const int b = owner(bk, B, i);
            a.free_pages[count + i] = a.table[(size_t)b * a.max_pages + i - bk[b]];
        }
    }
    if (bk[B] > 0) __syncthreads();                    // the free list is read, and bk written, below
    for (int b = b0; b < b1; ++b) {
        const int len = length(b), add = a.add[b];
        const bool served = add > 0 && (long long)len + add <= most && st[b + 1] <= a.max_tokens &&
                            (nd[b + 1] == nd[b] || nd[b + 1] <= F);
        a.lengths_out[b] = add < 0 ? 0 : (served ? len + add : len);
        if (served && nd[b + 1] > nd[b]) atomicMax(&s_taken, nd[b + 1]);
        if (add > 0 && !served) atomicAdd(&s_refused, 1);
        if (!rows_here && add > 0 && st[b] < a.max_tokens) a.positions[st[b]] = served ? len : -1;
        bk[b] = served ? len : -1;
    }
    __syncthreads();
    const int taken = s_taken;
    for (int m = tid; m < taken; m += THREADS) {
        const int b = owner(nd, B, m);
        a.table[(size_t)b * a.max_pages + pages_of(bk[b], a.shift) + m - nd[b]] = a.free_pages[F - 1 - m];
    }
    if (tid == 0) {
        *a.free_count_out = F - taken;
        *a.refused = s_refused;
    }
    if (!rows_here) return;
    // a row's page: one that the request had, or one taken above (from the free list: the table entry may be on its way)
    const int T = st[B];
    for (int t = tid; t < a.max_tokens; t += THREADS) {
        int pos = -1, page = -1;
        if (t < T) {
            const int b = owner(st, B, t);
            if (bk[b] >= 0) {
                pos = bk[b] + t - st[b];
                const int fresh = (pos >> a.shift) - pages_of(bk[b], a.shift);
                page = fresh >= 0 ? a.free_pages[F - 1 - nd[b] - fresh] : a.table[(size_t)b * a.max_pages + (pos >> a.shift)];
            }
        }
        write_row(a, t, pos, page);
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
    int pos = -1, page = -1;
    if (t < a.starts[a.B]) {
        const int b = owner(a.starts, a.B, t), s = a.starts[b], first = a.positions[s];
        if (first >= 0) {
            pos = first + t - s;
            page = a.table[(size_t)b * a.max_pages + (pos >> a.shift)];
        }
    }
    write_row(a, t, pos, page);
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t st)
{
    const size_t smem = (size_t)3 * (a.B + 1) * sizeof(int);
    const int rows_here = a.max_tokens <= kRowsInPlan;
    cudaError_t e = cudaSuccess;
    if (a.B <= kFew && a.max_tokens <= kFew) {
        page_plan_kernel<128><<<1, 128, smem, st>>>(a, rows_here);
    } else {
        if (smem > 48 * 1024)
            e = cudaFuncSetAttribute(page_plan_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        page_plan_kernel<1024><<<1, 1024, smem, st>>>(a, rows_here);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess || rows_here) return e;
    return launch_pdl(page_rows_kernel, dim3((unsigned)((a.max_tokens + kRowThreads - 1) / kRowThreads)),
                      dim3(kRowThreads), 0, st, a);
}

}  // namespace fadkv
