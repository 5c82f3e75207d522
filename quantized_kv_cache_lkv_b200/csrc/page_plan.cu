// page_plan.cu -- block tables, lengths and slot maps from request lengths
// (lkv_page_plan).
//
// need_b = ceil((len_b + new_b) / 256) - ceil(len_b / 256) pages; prefix sums
// of new_b and need_b over the sequences give every token its row and every
// new page its entry of the free stack, and cut the batch where the first
// sequence does not fit (both sums rise, so those that fit come first).
//
// Latency bound: a decode step moves a few hundred bytes.  So one launch, and
// no step that waits for another block: every block builds both prefix sums
// itself in shared memory (the lengths come out of L2), and a token on a new
// page takes the page from the free stack rather than from the table entry
// that some other block is writing.
#include <algorithm>

#include "serving.cuh"

namespace lkv {

namespace {

constexpr int kThreads = 512;

// Saturating sum of non-negative ints: past any capacity, but never wrapped.
__device__ __forceinline__ int add_sat(int a, int b) {
  const unsigned s = (unsigned)a + (unsigned)b;
  return s > 0x7FFFFFFFu ? 0x7FFFFFFF : (int)s;
}

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPageTokens - 1) / kPageTokens; }

__device__ __forceinline__ bool sane(const PlanArgs& a, int len, int add) {
  return len >= 0 && add >= 0 && (long long)len + add <= (long long)a.pps * kPageTokens;
}

// Last b of [0, n) with first[b] <= x (first[0] = 0 <= x < first[n]).
__device__ __forceinline__ int owner(const int* first, int n, int x, int most) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (min(first[mid], most) <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(PlanArgs a) {
  extern __shared__ int s_tok[];       // [B + 1] tokens before each sequence
  int* s_pg = s_tok + a.B + 1;         // [B + 1] new pages before each sequence
  __shared__ int s_wt[32], s_wp[32], s_cut[2], s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int count = clamp_len(__ldg(a.free_count), a.free_cap);
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  if (tid < 2) s_cut[tid] = 0;
  if (tid == 2) s_bad = 0;
  int nt = 0, np = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int len = __ldg(a.lens + b), add = __ldg(a.n_new + b);
    const bool ok = sane(a, len, add);
    const int t = ok ? add : 0, p = ok ? pages_of(len + add) - pages_of(len) : 0;
    bad |= !ok;
    nt = add_sat(nt, t);
    np = add_sat(np, p);
    s_tok[b + 1] = nt;  // within the thread's run for now
    s_pg[b + 1] = np;
  }
  int it = nt, ip = np;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, it, off), y = __shfl_up_sync(0xFFFFFFFFu, ip, off);
    if (lane >= off) { it = add_sat(it, x); ip = add_sat(ip, y); }
  }
  if (lane == 31) { s_wt[warp] = it; s_wp[warp] = ip; }
  __syncthreads();
  // exclusive sums before this thread's run
  int et = __shfl_up_sync(0xFFFFFFFFu, it, 1), ep = __shfl_up_sync(0xFFFFFFFFu, ip, 1);
  if (lane == 0) et = ep = 0;
  for (int w = 0; w < warp; ++w) { et = add_sat(et, s_wt[w]); ep = add_sat(ep, s_wp[w]); }
  int ct = 0, cp = 0;
  for (int b = b0; b < b1; ++b) {
    const int t = add_sat(s_tok[b + 1], et), p = add_sat(s_pg[b + 1], ep);
    s_tok[b + 1] = t;
    s_pg[b + 1] = p;
    if (t <= a.n_cap && p <= count) { ct = t; cp = p; } else { bad = true; }
  }
  if (tid == 0) s_tok[0] = s_pg[0] = 0;
  if (ct) atomicMax(&s_cut[0], ct);
  if (cp) atomicMax(&s_cut[1], cp);
  if (bad) s_bad = 1;
  __syncthreads();
  // everything behind the cut counts as nothing: min() with these two
  const int tokens = s_cut[0], pages = s_cut[1];
  const int gt = blockIdx.x * kThreads + tid, gn = gridDim.x * kThreads;
  for (int b = gt; b < a.B; b += gn) {
    const int t0 = min(s_tok[b], tokens), t1 = min(s_tok[b + 1], tokens);
    a.new_lens[b] = __ldg(a.lens + b) + (t1 - t0);
    a.cu[b + 1] = t1;
  }
  for (int k = gt; k < pages; k += gn) {
    const int b = owner(s_pg, a.B, k, pages);
    const int j = pages_of(__ldg(a.lens + b)) + k - s_pg[b];
    a.table[(long long)b * a.pps + j] = __ldg(a.free_pages + count - 1 - k);
  }
  for (int t = gt; t < tokens; t += gn) {
    const int b = owner(s_tok, a.B, t, tokens);
    const int len = __ldg(a.lens + b), old = pages_of(len);
    const int pos = len + t - s_tok[b];
    const int j = pos / kPageTokens;
    const int page = j < old ? a.table[(long long)b * a.pps + j] : __ldg(a.free_pages + count - 1 - (s_pg[b] + j - old));
    a.positions[t] = pos;
    a.token_seq[t] = b;
    a.slots[t] = page >= 0 && page < a.num_pages ? (long long)page * kPageTokens + pos % kPageTokens : -1;
  }
  if (blockIdx.x != gridDim.x - 1) return;
  // the last block also answers for the call: every page a new token can lie
  // on is a taken one or the last old page of a served sequence
  if (tid == 0) { a.cu[0] = 0; a.free_left[0] = count - pages; }
  if (a.status == nullptr) return;
  bad = false;
  for (int k = tid; k < pages; k += kThreads) {
    const int page = __ldg(a.free_pages + count - 1 - k);
    bad |= page < 0 || page >= a.num_pages;
  }
  for (int b = tid; b < a.B; b += kThreads) {
    const int len = __ldg(a.lens + b);
    if (min(s_tok[b + 1], tokens) > min(s_tok[b], tokens) && len % kPageTokens != 0) {
      const int page = a.table[(long long)b * a.pps + len / kPageTokens];
      bad |= page < 0 || page >= a.num_pages;
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (tid == 0) a.status[0] = s_bad ? kStatusInvalidArg : 0;
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)2 * (a.B + 1) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const long long want = ((long long)std::max(a.n_cap, a.B) + kThreads - 1) / kThreads;
  const int grid = (int)std::max<long long>(1, std::min<long long>(num_sms(), want));
  page_plan_kernel<<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace lkv
