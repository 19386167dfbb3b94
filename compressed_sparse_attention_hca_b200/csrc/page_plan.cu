// page_plan.cu -- block tables and slot maps of a step from the requests'
// lengths (admirer.cn article, cache paragraph: compressed rows in fixed pages
// of 128 tokens taken from a shared pool).
//
// Everything a page or a slot needs follows from exclusive prefix sums over
// the requests: pages taken, pages given back, new rows of each cache.  Every
// CTA forms these sums itself (16 bytes a request, from L2 after the first
// CTA), then takes its share of the outputs: slots of the new rows, table
// slots of the pages taken, stack places of the pages given back.  A new
// page's number is read from the stack (or from the table slot of the page
// given back that lies there), never from what another CTA writes, so the CTAs
// do not wait for one another; the stack's count, if updated in place,
// is written by the last CTA to have read it.
//
// Places of the table that hold no page (the stack was empty when they were
// taken) are not given back, so every CTA first counts the pages that are: of a
// request that gives back a few places the thread that reads its lengths, of
// one that gives back many all warps, 256 places at a time.
//
// Latency bounds it: a step of 256 requests takes 6.4 us (a launch ~2.5, then
// four or five dependent reads and the scan), one that rolls back 4.4 (4.1
// without the count of pages), 16 prompts of 131,072 to 262,144 tokens 14.2 us
// for 8 MB of slots (13.6).  Code comes cold from the instruction cache, so loops are
// not unrolled (the compiler's choice took 4 to 9 % longer).
#include "csa_internal.cuh"
#include "sm100.cuh"

namespace csa {

CSA_DEFINE_STATUS_READER(take_status_page_plan)

namespace {

constexpr int kThreads = 256;
constexpr int kFew = 4;    // places given back that a thread looks at by itself
constexpr int kAhead = 8;  // reads of places that a lane has in flight where there are more
constexpr int64_t kMaxLen = (int64_t)1 << 40;

__device__ __forceinline__ int64_t clamp_len(int64_t n) { return n < 0 ? 0 : min64(n, kMaxLen); }
// x / d for 0 <= x <= 2^41, d <= 2^20, with inv = ceil(2^64 / d) (0 for d = 1):
// floor(x inv / 2^64) is exact, as it exceeds x / d by x (inv d - 2^64) / (d 2^64) < 2^-23 < 1 / d.
// A 64-bit division takes ~100 dependent instructions, and a step of 256
// requests spent most of its 16 us in them.
__device__ __forceinline__ int64_t quot(int64_t x, uint64_t inv) {
  return inv == 0 ? x : (int64_t)__umul64hi((uint64_t)x, inv);
}
__device__ __forceinline__ int64_t pages_of(int64_t n, const PagePlanArgs& a) {
  return quot(n + a.page_tokens - 1, a.inv_page);
}

// The sums of one request (or of several).
struct Sums {
  int take, give;
  int64_t rows[kMaxSlotMaps], want;
  __device__ __forceinline__ void add(const Sums& o) {
    take += o.take;
    give += o.give;
    want += o.want;
#pragma unroll
    for (int i = 0; i < kMaxSlotMaps; ++i) rows[i] += o.rows[i];
  }
  __device__ __forceinline__ Sums shfl_up(int d) const {
    Sums r;
    r.take = __shfl_up_sync(0xffffffffu, take, d);
    r.give = __shfl_up_sync(0xffffffffu, give, d);
    r.want = __shfl_up_sync(0xffffffffu, want, d);
#pragma unroll
    for (int i = 0; i < kMaxSlotMaps; ++i) r.rows[i] = __shfl_up_sync(0xffffffffu, rows[i], d);
    return r;
  }
};

// All of a request's sums but the pages given back, which lie in [p1, p0).
__device__ __forceinline__ Sums sums_of(const PagePlanArgs& a, int b, int* p0_out, int* p1_out) {
  const int64_t before = clamp_len(a.len_before[b]), after = clamp_len(a.len_after[b]);
  const int64_t p0 = min64(pages_of(before, a), a.max_pages), want = pages_of(after, a);
  const int64_t p1 = min64(want, a.max_pages);
  Sums s;
  s.take = (int)max64(0, p1 - p0);
  s.give = 0;
  s.want = max64(0, want - p0);
#pragma unroll
  for (int i = 0; i < kMaxSlotMaps; ++i)
    s.rows[i] = i < a.n_maps ? max64(0, quot(after, a.maps[i].inv_m) - quot(before, a.maps[i].inv_m)) : 0;
  *p0_out = (int)p0;
  *p1_out = (int)p1;
  return s;
}

// The request whose range [pre[b], pre[b + 1]) holds x (x < pre[batch]).
template <class T>
__device__ __forceinline__ int owner(const T* pre, int batch, T x) {
  int lo = 0, hi = batch;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ bool is_page(const PagePlanArgs& a, int pg) { return (uint32_t)pg < (uint32_t)a.n_pages; }
// What is neither a page nor the -1 of one that could not be had.
__device__ __forceinline__ bool is_bad(const PagePlanArgs& a, int pg) { return pg != -1 && !is_page(a, pg); }
// The k-th place from `at` on that holds a page (`last` if there are fewer).
__device__ __forceinline__ const int32_t* nth_page(const PagePlanArgs& a, const int32_t* at, const int32_t* last, int k) {
#pragma unroll 1
  for (; at < last; ++at)
    if (is_page(a, *at) && k-- == 0) break;
  return at;
}

// Where a thread has got to among a request's places that do not all hold a page.
struct Cursor {
  int b = -1, k;  // page k of request b
  const int32_t* at;
};

struct Plan {
  const PagePlanArgs& a;
  const int *take, *give;  // prefix sums [batch + 1] of places taken and pages given back
  const int *p0, *p1;      // pages before and after [batch]
  int count, R;
  // The page at `at`, -1 where there is none.
  __device__ __forceinline__ int checked(const int32_t* at) const {
    if (at == nullptr) return -1;
    const int pg = *at;
    if (is_page(a, pg)) return pg;
    if (pg != -1 || (at >= a.free_list && at < a.free_list + a.n_pages)) flag_status(kStatusBadPage);
    return -1;
  }
  // The place of the i-th page given back.
  __device__ __forceinline__ const int32_t* given(int i, Cursor& c) const {
    const int b = owner(give, a.batch, i), k = i - give[b], n = p0[b] - p1[b];
    const int32_t* const row = a.table + (int64_t)b * a.max_pages + p1[b];
    if (give[b + 1] - give[b] == n) return row + k;
    const bool on = c.b == b && c.k < k;
    c.at = nth_page(a, on ? c.at + 1 : row, row + n - 1, on ? k - c.k - 1 : k);
    c.b = b;
    c.k = k;
    return c.at;
  }
  // Where the number of page i of the pages taken is read: in the stack, or in
  // the table slot of the page given back that this call puts there; nullptr
  // when the stack is empty by then.
  __device__ __forceinline__ const int32_t* taken(int64_t i) const {
    if (i < R) {
      Cursor c;
      return given((int)i, c);
    }
    const int64_t at = (int64_t)count + R - 1 - i;
    return at < 0 ? nullptr : a.free_list + at;
  }
  // The same for page j of request b after the step; nullptr when it has none.
  __device__ __forceinline__ const int32_t* page(int b, int64_t j) const {
    if (j < p0[b]) return a.table + (int64_t)b * a.max_pages + j;
    const int64_t i = (int64_t)take[b] + (j - p0[b]);
    return i < take[b + 1] ? taken(i) : nullptr;
  }
};

// The page numbers that slot i of a map needs, and the row they are for.
struct SlotAt {
  int b;
  int64_t r, j;
  __device__ __forceinline__ SlotAt(const Plan& p, const SlotMap& m, const int64_t* pre, int64_t i)
      : b(owner(pre, p.a.batch, i)),
        r(quot(clamp_len(p.a.len_before[b]), m.inv_m) + (i - pre[b])),
        j(quot(r, m.inv_rows)) {}
};

// Slots i .. i + VEC - 1 of a map (VEC of them exist).  Steps of few rows a
// request take a slot per thread: its page is two dependent reads away, and
// four such chains one after the other in a thread took twice the whole step's
// time.  Prompts take four, which mostly share a page and are stored at once.
template <int VEC>
__device__ __forceinline__ void write_slots(const Plan& p, const SlotMap& m, const int64_t* pre, int64_t i0) {
  int slot[VEC], sf[VEC];
#pragma unroll
  for (int u = 0; u < VEC; ++u) slot[u] = sf[u] = -1;
  const int64_t total = pre[p.a.batch];
  if (i0 < total) {
    const SlotAt s(p, m, pre, i0);
    // one lookup serves the slots of the same request, page and 128 rows
    const int64_t in_page = m.page_rows - (s.r - s.j * m.page_rows), in_block = 128 - (s.r & 127);
    int64_t same = min64(pre[s.b + 1] - i0, in_page);
    if (m.sf_slots != nullptr) same = min64(same, in_block);
    int u = 0;
    SlotAt t = s;
    for (;;) {
      const int32_t* at = p.page(t.b, t.j);
      const int32_t* sf_at = m.sf_slots != nullptr ? p.page(t.b, quot(t.r & ~(int64_t)127, m.inv_rows)) : nullptr;
      const int pg = p.checked(at), sf_pg = p.checked(sf_at);
      const int slot0 = pg * m.page_rows + (int)(t.r - t.j * m.page_rows), sf0 = sf_pg * 128 + (int)(t.r & 127);
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if (v >= u && v - u < same && pg >= 0) {
          slot[v] = slot0 + v - u;
          if (sf_pg >= 0) sf[v] = sf0 + v - u;
        }
      if (u + same >= VEC || i0 + u + same >= total) break;
      u += (int)same;
      t = SlotAt(p, m, pre, i0 + u);
      same = 1;
    }
  }
  if (VEC == 4) {
    *reinterpret_cast<int4*>(m.slots + i0) = make_int4(slot[0], slot[VEC > 1], slot[VEC / 2], slot[VEC - 1]);
    if (m.sf_slots != nullptr)
      *reinterpret_cast<int4*>(m.sf_slots + i0) = make_int4(sf[0], sf[VEC > 1], sf[VEC / 2], sf[VEC - 1]);
  } else {
    m.slots[i0] = slot[0];
    if (m.sf_slots != nullptr) m.sf_slots[i0] = sf[0];
  }
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(PagePlanArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  int64_t* row_pre = reinterpret_cast<int64_t*>(smem);  // [n_maps][batch + 1]
  int* take = reinterpret_cast<int*>(row_pre + (int64_t)a.n_maps * (a.batch + 1));
  int* give = take + a.batch + 1;
  int* p0 = give + a.batch + 1;
  int* p1 = p0 + a.batch;
  __shared__ Sums warp_sums[kThreads / 32];
  __shared__ int64_t want_total;
  __shared__ int n_long;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) n_long = 0;
  __syncthreads();
  after_previous();
  const int c0 = *a.count;
  const int count = (int)max64(0, min64(c0, a.n_pages));

  // the sums of a run of requests per thread; give[b]: the pages that b gives back
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  Sums mine{};
  bool bad = false;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    mine.add(sums_of(a, b, &p0[b], &p1[b]));
    const int n = p0[b] - p1[b];
    int pages = 0;
    if (n > kFew) {
      take[atomicAdd(&n_long, 1)] = b;  // a list of them, until the prefix sums replace it
    } else if (n > 0) {
      const int32_t* const row = a.table + (int64_t)b * a.max_pages + p1[b];
      int pg[kFew];
#pragma unroll
      for (int j = 0; j < kFew; ++j) pg[j] = row[min(j, n - 1)];
#pragma unroll
      for (int j = 0; j < kFew; ++j) {
        pages += j < n && is_page(a, pg[j]);
        bad |= is_bad(a, pg[j]);
      }
    }
    give[b] = pages;
  }
  __syncthreads();
  int turn = 0;  // of the warps
#pragma unroll 1
  for (int l = 0; l < n_long; ++l) {
    const int b = take[l];
    const uint32_t n = (uint32_t)(p0[b] - p1[b]);
    const int32_t* const row = a.table + (int64_t)b * a.max_pages + p1[b];
#pragma unroll 1
    for (uint32_t j0 = 0; j0 < n; j0 += 32 * kAhead, ++turn) {
      if (turn % (kThreads / 32) != warp) continue;
      int pg[kAhead], pages = 0;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) pg[u] = row[min(j0 + 32 * u + lane, n - 1)];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        pages += j0 + 32 * u + lane < n && is_page(a, pg[u]);
        bad |= is_bad(a, pg[u]);
      }
      pages = __reduce_add_sync(0xffffffffu, pages);
      if (lane == 0) atomicAdd(&give[b], pages);
    }
  }
  if (n_long > 0) __syncthreads();
  if (bad) flag_status(kStatusBadPage);
  // exclusive prefix sums: over lanes, then warps, then the thread's requests
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine.give += give[b];
  Sums inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = inc.shfl_up(d);
    if (lane >= d) inc.add(o);
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  Sums run{};
#pragma unroll 1
  for (int w = 0; w < warp; ++w) run.add(warp_sums[w]);
  const Sums before_lane = inc.shfl_up(1);
  if (lane > 0) run.add(before_lane);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    int q0, q1;
    Sums s = sums_of(a, b, &q0, &q1);
    s.give = give[b];
    take[b] = run.take;
    give[b] = run.give;
    for (int i = 0; i < a.n_maps; ++i) row_pre[i * (a.batch + 1) + b] = run.rows[i];
    run.add(s);
  }
  if (tid == kThreads - 1) {  // its run ends at the last request
    take[a.batch] = run.take;
    give[a.batch] = run.give;
    for (int i = 0; i < a.n_maps; ++i) row_pre[i * (a.batch + 1) + a.batch] = run.rows[i];
    want_total = run.want;
  }
  __syncthreads();

  const int A = take[a.batch], R = give[a.batch];
  const Plan plan{a, take, give, p0, p1, count, R};
  const int64_t t0 = (int64_t)blockIdx.x * kThreads + tid, nt = (int64_t)gridDim.x * kThreads;
#pragma unroll 1
  for (int i = 0; i < a.n_maps; ++i) {
    const SlotMap& m = a.maps[i];
    const int64_t* pre = row_pre + i * (a.batch + 1);
    const int64_t quads = m.capacity >= 128 * (int64_t)a.batch ? m.capacity / 4 : 0;
#pragma unroll 1
    for (int64_t s = t0; s < quads; s += nt) write_slots<4>(plan, m, pre, 4 * s);
#pragma unroll 1
    for (int64_t s = 4 * quads + t0; s < m.capacity; s += nt) write_slots<1>(plan, m, pre, s);
    if (blockIdx.x == 0)
#pragma unroll 1
      for (int b = tid; b <= a.batch; b += kThreads) m.row_start[b] = pre[b];
  }
#pragma unroll 1
  for (int64_t i = t0; i < A; i += nt) {
    const int b = owner(take, a.batch, (int)i);
    a.table[(int64_t)b * a.max_pages + p0[b] + (i - take[b])] = plan.checked(plan.taken(i));
  }
  Cursor c;
#pragma unroll 1
  for (int64_t i = t0; i < R; i += nt) {
    const int64_t at = (int64_t)count + R - 1 - i;
    if (at < a.n_pages) a.free_list[at] = *plan.given((int)i, c);
    else flag_status(kStatusBadPage);
  }

  // a count updated in place is written by the last CTA, when every one has
  // read it; another place by the first
  const bool in_place = a.count == a.count_out && gridDim.x > 1;
  if (in_place) __syncthreads();
  if (tid == 0) {
    bool last = blockIdx.x == 0;
    if (in_place) {
      __threadfence();
      last = atomicAdd(a.info + 3, 1) == (int)gridDim.x - 1;
    }
    if (last) {
      const int got = (int)min64(A, (int64_t)count + R);
      *a.count_out = (int)min64((int64_t)count + R - got, a.n_pages);
      a.info[0] = got;
      a.info[1] = R;
      a.info[2] = (int)min64(want_total - got, 0x7FFFFFFF);
      a.info[3] = 0;
      if (c0 != count) flag_status(kStatusBadPage);
    }
  }
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs& args, cudaStream_t s) {
  PagePlanArgs a = args;
  const auto inverse = [](int d) { return d <= 1 ? 0 : ~(uint64_t)0 / (uint64_t)d + 1; };  // ceil(2^64 / d)
  a.inv_page = inverse(a.page_tokens);
  for (int i = 0; i < a.n_maps; ++i) {
    a.maps[i].inv_m = inverse(a.maps[i].m);
    a.maps[i].inv_rows = inverse(a.maps[i].page_rows);
  }
  const size_t smem = (size_t)(a.batch + 1) * (8 * a.n_maps + 16);
  if (smem > 40 * 1024) {  // 48 KB without asking, the kernel's static arrays among them
    const cudaError_t e =
        cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  int64_t work = 1;  // threads that have something to do at once
  for (int i = 0; i < a.n_maps; ++i)
    work = max64(work, a.maps[i].capacity >= 128 * (int64_t)a.batch ? a.maps[i].capacity / 4 : a.maps[i].capacity);
  const int64_t blocks = min64((work + kThreads - 1) / kThreads, 3 * 148);
  return launch_overlapped(page_plan_kernel, (unsigned)blocks, kThreads, smem, 1, s, a);
}

}  // namespace csa
